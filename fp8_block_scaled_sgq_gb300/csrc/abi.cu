// C-ABI entry points: argument validation, then the kernel launchers.
// Every check happens on the host before anything is enqueued; nothing
// aborts or falls back.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <mutex>

#include "sgq_internal.h"

namespace sgq {
namespace {

std::atomic<uint64_t> g_launches{0};
DeviceInfo g_dev[64];
bool g_dev_ok[64] = {};
std::mutex g_dev_mu;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned_to(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// The latent-attention calls: element type, rotated width (whole 16-byte
// columns of pairs), strides (16-byte columns).
bool good_dtype(int dtype) { return dtype == SGQ_BF16 || dtype == SGQ_FP16; }
bool good_rotation(int R, int interleaved) {
    return (interleaved == 0 || interleaved == 1) && R > 0 && R <= 2048 && R % (interleaved ? 8 : 16) == 0;
}
bool good_strides(std::initializer_list<int64_t> strides) {
    for (const int64_t s : strides)
        if (s < 0 || s % 8 != 0 || s > (int64_t(1) << 40)) return false;
    return true;
}
// Tokens and heads of the absorbed attention: fewer than 2^31 rows (tokens
// first, so that the product does not wrap).
bool good_rows(int64_t T, int64_t H) {
    return T >= 0 && T < (int64_t(1) << 31) && H > 0 && H <= 65535 && T * H < (int64_t(1) << 31);
}

}  // namespace

void note_launch(int n) { g_launches.fetch_add(static_cast<uint64_t>(n), std::memory_order_relaxed); }

sgq_status device_info(DeviceInfo* out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SGQ_ERR_CUDA;
    std::lock_guard<std::mutex> lk(g_dev_mu);
    if (!g_dev_ok[dev]) {
        DeviceInfo d;
        if (cudaDeviceGetAttribute(&d.sm_count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&d.max_smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) !=
                cudaSuccess ||
            cudaDeviceGetAttribute(&d.cc_major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&d.cc_minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
            return SGQ_ERR_CUDA;
        g_dev[dev] = d;
        g_dev_ok[dev] = true;
    }
    *out = g_dev[dev];
    return SGQ_OK;
}

}  // namespace sgq

using sgq::aligned16;
using sgq::aligned_to;
using sgq::good_dtype;
using sgq::good_rotation;
using sgq::good_rows;
using sgq::good_strides;

extern "C" {

sgq_status sgq_quant_token_group(const void* x, int64_t M, int64_t K, int group, int ue8m0, void* xq,
                                 float* xs, sgq_stream_t stream) {
    if (M < 0 || K <= 0 || (group != 32 && group != 128) || K % group != 0 || (ue8m0 != 0 && ue8m0 != 1))
        return SGQ_ERR_INVALID_ARG;
    if (M > (int64_t(1) << 31) / 1 || M * K > (int64_t(1) << 40)) return SGQ_ERR_INVALID_ARG;
    if (M == 0) return SGQ_OK;
    if (!x || !xq || !xs) return SGQ_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(xq) || !aligned16(xs)) return SGQ_ERR_MISALIGNED;
    return sgq::launch_quant_token_group(x, M, K, group, ue8m0, xq, xs,
                                         reinterpret_cast<cudaStream_t>(stream));
}

sgq_status sgq_quant_token_group_ue8m0(const void* x, int64_t M, int64_t K, int group, void* xq, uint8_t* xe,
                                       sgq_stream_t stream) {
    if (M < 0 || K <= 0 || (group != 32 && group != 128) || K % group != 0) return SGQ_ERR_INVALID_ARG;
    if (M > (int64_t(1) << 31) / 1 || M * K > (int64_t(1) << 40)) return SGQ_ERR_INVALID_ARG;
    if (M == 0) return SGQ_OK;
    if (!x || !xq || !xe) return SGQ_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(xq) || !aligned16(xe)) return SGQ_ERR_MISALIGNED;
    return sgq::launch_quant_token_group_e8(x, M, K, group, xq, xe, reinterpret_cast<cudaStream_t>(stream));
}

sgq_status sgq_scales_to_ue8m0(const float* s, int64_t n, uint8_t* e, sgq_stream_t stream) {
    if (n < 0 || n > (int64_t(1) << 40)) return SGQ_ERR_INVALID_ARG;
    if (n == 0) return SGQ_OK;
    if (!s || !e) return SGQ_ERR_INVALID_ARG;
    return sgq::launch_scales_to_ue8m0(s, n, e, reinterpret_cast<cudaStream_t>(stream));
}

sgq_status sgq_quant_weight_block(const void* w, int64_t N, int64_t K, int blk_n, int blk_k, int ue8m0,
                                  void* wq, float* ws, sgq_stream_t stream) {
    if (N < 0 || K <= 0 || (blk_n != 32 && blk_n != 128) || (blk_k != 32 && blk_k != 128) ||
        K % blk_k != 0 || (ue8m0 != 0 && ue8m0 != 1))
        return SGQ_ERR_INVALID_ARG;
    if ((N + blk_n - 1) / blk_n > 65535 || K / blk_k > (int64_t(1) << 31) - 1) return SGQ_ERR_INVALID_ARG;
    if (N == 0) return SGQ_OK;
    if (!w || !wq || !ws) return SGQ_ERR_INVALID_ARG;
    if (!aligned16(w) || !aligned16(wq) || !aligned16(ws)) return SGQ_ERR_MISALIGNED;
    return sgq::launch_quant_weight_block(w, N, K, blk_n, blk_k, ue8m0, wq, ws,
                                          reinterpret_cast<cudaStream_t>(stream));
}

sgq_status sgq_fp8_block_gemm_ex(const void* Aq, const float* As, const void* Wq, const float* Ws, void* D,
                                 int64_t M, int64_t N, int64_t K, int blk_n, int blk_k, uint32_t flags,
                                 sgq_stream_t stream) {
    if (M < 0 || N <= 0 || K <= 0 || (blk_n != 32 && blk_n != 128) || (blk_k != 32 && blk_k != 128) ||
        K % blk_k != 0 || N % 8 != 0 ||
        (flags & ~uint32_t(SGQ_GEMM_FORCE_PROMOTE | SGQ_GEMM_ISSUE_ALT | SGQ_GEMM_ISSUE_SINGLE |
                           SGQ_GEMM_TEST_TIMEOUT | SGQ_GEMM_SCALES_POW2)) != 0 ||
        (flags & (SGQ_GEMM_ISSUE_ALT | SGQ_GEMM_ISSUE_SINGLE)) == (SGQ_GEMM_ISSUE_ALT | SGQ_GEMM_ISSUE_SINGLE))
        return SGQ_ERR_INVALID_ARG;
    // int32 indexing inside the kernel
    if (M >= (int64_t(1) << 31) || N >= (int64_t(1) << 31) || K >= (int64_t(1) << 31))
        return SGQ_ERR_INVALID_ARG;
    if (M == 0) return SGQ_OK;
    if (!Aq || !As || !Wq || !Ws || !D) return SGQ_ERR_INVALID_ARG;
    if (!aligned16(Aq) || !aligned16(As) || !aligned16(Wq) || !aligned16(Ws) || !aligned16(D))
        return SGQ_ERR_MISALIGNED;
    return sgq::launch_fp8_block_gemm(Aq, As, Wq, Ws, D, M, N, K, blk_n, blk_k, flags,
                                      reinterpret_cast<cudaStream_t>(stream));
}

sgq_status sgq_fp8_block_gemm(const void* Aq, const float* As, const void* Wq, const float* Ws, void* D,
                              int64_t M, int64_t N, int64_t K, int blk_n, int blk_k, sgq_stream_t stream) {
    return sgq_fp8_block_gemm_ex(Aq, As, Wq, Ws, D, M, N, K, blk_n, blk_k, SGQ_GEMM_DEFAULT, stream);
}

sgq_status sgq_fp8_block_gemm_ue8m0(const void* Aq, const uint8_t* Ae, const void* Wq, const uint8_t* We, void* D,
                                    int64_t M, int64_t N, int64_t K, int blk_n, int blk_k, uint32_t flags,
                                    sgq_stream_t stream) {
    if (M < 0 || N <= 0 || K <= 0 || (blk_n != 32 && blk_n != 128) || (blk_k != 32 && blk_k != 128) ||
        K % blk_k != 0 || N % 8 != 0 ||
        (flags & ~uint32_t(SGQ_GEMM_FORCE_PROMOTE | SGQ_GEMM_ISSUE_ALT | SGQ_GEMM_ISSUE_SINGLE |
                           SGQ_GEMM_SCALES_POW2)) != 0 ||
        (flags & (SGQ_GEMM_ISSUE_ALT | SGQ_GEMM_ISSUE_SINGLE)) == (SGQ_GEMM_ISSUE_ALT | SGQ_GEMM_ISSUE_SINGLE))
        return SGQ_ERR_INVALID_ARG;
    if (M >= (int64_t(1) << 31) || N >= (int64_t(1) << 31) || K >= (int64_t(1) << 31))
        return SGQ_ERR_INVALID_ARG;
    if (M == 0) return SGQ_OK;
    if (!Aq || !Ae || !Wq || !We || !D) return SGQ_ERR_INVALID_ARG;
    if (!aligned16(Aq) || !aligned16(Ae) || !aligned16(Wq) || !aligned16(We) || !aligned16(D))
        return SGQ_ERR_MISALIGNED;
    return sgq::launch_fp8_block_gemm_ue8m0(Aq, Ae, Wq, We, D, M, N, K, blk_n, blk_k, flags,
                                            reinterpret_cast<cudaStream_t>(stream));
}

sgq_status sgq_fp8_block_gemm_noalloc(const void* Aq, const float* As, const void* Wq, const float* Ws,
                                      void* D, int64_t M, int64_t N, int64_t K, int blk_n, int blk_k,
                                      sgq_stream_t stream) {
    if (M < 0 || N <= 0 || K <= 0 || (blk_n != 32 && blk_n != 128) || (blk_k != 32 && blk_k != 128) ||
        K % blk_k != 0 || N % 8 != 0)
        return SGQ_ERR_INVALID_ARG;
    if (M >= (int64_t(1) << 31) || N >= (int64_t(1) << 31) || K >= (int64_t(1) << 31))
        return SGQ_ERR_INVALID_ARG;
    if (M == 0) return SGQ_OK;
    if (!Aq || !As || !Wq || !Ws || !D) return SGQ_ERR_INVALID_ARG;
    if (!aligned16(Aq) || !aligned16(As) || !aligned16(Wq) || !aligned16(Ws) || !aligned16(D))
        return SGQ_ERR_MISALIGNED;
    return sgq::launch_fp8_block_gemm_noalloc(Aq, As, Wq, Ws, D, M, N, K, blk_n, blk_k,
                                              reinterpret_cast<cudaStream_t>(stream));
}

sgq_status sgq_quant_token_group_v2(const void* x, int64_t E, int64_t T, int64_t H, int group, int ue8m0,
                                    int fuse_silu_and_mul, const int32_t* masked_m, void* xq, float* xs,
                                    sgq_stream_t stream) {
    if (E < 0 || T < 0 || H <= 0 || (group != 32 && group != 128) || H % group != 0 ||
        (ue8m0 != 0 && ue8m0 != 1) || (fuse_silu_and_mul != 0 && fuse_silu_and_mul != 1))
        return SGQ_ERR_INVALID_ARG;
    if (E >= (int64_t(1) << 31) || T >= (int64_t(1) << 31) || E * T * H > (int64_t(1) << 40))
        return SGQ_ERR_INVALID_ARG;
    if (E == 0 || T == 0) return SGQ_OK;
    if (!x || !xq || !xs) return SGQ_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(xq) || !aligned16(xs) || (masked_m && !aligned16(masked_m)))
        return SGQ_ERR_MISALIGNED;
    return sgq::launch_quant_token_group_v2(x, E, T, H, group, ue8m0, fuse_silu_and_mul, masked_m, xq, xs,
                                            reinterpret_cast<cudaStream_t>(stream));
}

sgq_status sgq_quant_per_token(const void* x, int64_t M, int64_t K, void* xq, float* xs, sgq_stream_t stream) {
    if (M < 0 || K <= 0 || K % 16 != 0 || M >= (int64_t(1) << 31) || M * K > (int64_t(1) << 40))
        return SGQ_ERR_INVALID_ARG;
    if (M == 0) return SGQ_OK;
    if (!x || !xq || !xs) return SGQ_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(xq) || !aligned16(xs)) return SGQ_ERR_MISALIGNED;
    return sgq::launch_quant_per_token(x, M, K, xq, xs, reinterpret_cast<cudaStream_t>(stream));
}

sgq_status sgq_quant_per_tensor(const void* x, int64_t n, int is_static, void* xq, float* xs, sgq_stream_t stream) {
    if (n < 0 || n % 16 != 0 || n > (int64_t(1) << 40) || (is_static != 0 && is_static != 1))
        return SGQ_ERR_INVALID_ARG;
    if (n == 0) return SGQ_OK;
    if (!x || !xq || !xs) return SGQ_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(xq) || !aligned16(xs)) return SGQ_ERR_MISALIGNED;
    return sgq::launch_quant_per_tensor(x, n, is_static, xq, xs, reinterpret_cast<cudaStream_t>(stream));
}

sgq_status sgq_fp8_scaled_mm(const void* Aq, const float* sa, int64_t sa_n, const void* Wq, const float* sb,
                             int64_t sb_n, const void* bias, void* D, int64_t M, int64_t N, int64_t K,
                             sgq_stream_t stream) {
    if (M < 0 || N <= 0 || K <= 0 || K % 32 != 0 || N % 8 != 0) return SGQ_ERR_INVALID_ARG;
    if (M >= (int64_t(1) << 31) || N >= (int64_t(1) << 31) || K >= (int64_t(1) << 31)) return SGQ_ERR_INVALID_ARG;
    if ((sa_n != 1 && sa_n != M) || (sb_n != 1 && sb_n != N)) return SGQ_ERR_INVALID_ARG;
    if (M == 0) return SGQ_OK;
    if (!Aq || !sa || !Wq || !sb || !D) return SGQ_ERR_INVALID_ARG;
    if (!aligned16(Aq) || !aligned16(sa) || !aligned16(Wq) || !aligned16(sb) || !aligned16(D) ||
        (bias && !aligned16(bias)))
        return SGQ_ERR_MISALIGNED;
    return sgq::launch_fp8_scaled_mm(Aq, sa, sa_n, Wq, sb, sb_n, bias, D, M, N, K,
                                     reinterpret_cast<cudaStream_t>(stream));
}

sgq_status sgq_fp8_block_linear(const void* x, int ue8m0, const void* Wq, const float* Ws, void* D, int64_t M,
                                int64_t N, int64_t K, int blk_n, int blk_k, void* xq, float* xs,
                                sgq_stream_t stream) {
    if (M < 0 || N <= 0 || K <= 0 || (blk_n != 32 && blk_n != 128) || (blk_k != 32 && blk_k != 128) ||
        K % blk_k != 0 || N % 8 != 0 || (ue8m0 != 0 && ue8m0 != 1))
        return SGQ_ERR_INVALID_ARG;
    if (M >= (int64_t(1) << 31) || N >= (int64_t(1) << 31) || K >= (int64_t(1) << 31))
        return SGQ_ERR_INVALID_ARG;
    if ((xq == nullptr) != (xs == nullptr)) return SGQ_ERR_INVALID_ARG;
    if (M == 0) return SGQ_OK;
    if (!x || !Wq || !Ws || !D) return SGQ_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(Wq) || !aligned16(Ws) || !aligned16(D) || (xq && !aligned16(xq)) ||
        (xs && !aligned16(xs)))
        return SGQ_ERR_MISALIGNED;
    return sgq::launch_fp8_block_linear(x, ue8m0, Wq, Ws, D, M, N, K, blk_n, blk_k, xq, xs,
                                        reinterpret_cast<cudaStream_t>(stream));
}

sgq_status sgq_rotary(const void* x, int64_t T, int64_t H, int64_t D, int64_t x_stride_t, int64_t x_stride_h,
                      const int64_t* pos, const float* table, int64_t max_pos, int R, int64_t offset, int interleaved,
                      int inverse, int dtype, void* y, int64_t y_stride_t, int64_t y_stride_h, sgq_stream_t stream) {
    if (T < 0 || H < 0 || H > 65535 || D <= 0 || D > 2048 || D % 8 != 0 || max_pos <= 0 || offset < 0 || offset % 8 != 0 ||
        !good_rotation(R, interleaved) || offset + R > D || (inverse != 0 && inverse != 1) || !good_dtype(dtype) ||
        !good_strides({x_stride_t, x_stride_h, y_stride_t, y_stride_h}) || T >= (int64_t(1) << 31))
        return SGQ_ERR_INVALID_ARG;
    if (T == 0 || H == 0) return SGQ_OK;
    if (x == y && (x_stride_t != y_stride_t || x_stride_h != y_stride_h)) return SGQ_ERR_INVALID_ARG;
    if ((T > 1 && y_stride_t < D) || (H > 1 && y_stride_h < D)) return SGQ_ERR_INVALID_ARG;   // heads of y apart
    if (!x || !pos || !table || !y) return SGQ_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(table) || !aligned16(y) || !aligned_to(pos, 8)) return SGQ_ERR_MISALIGNED;
    return sgq::launch_rotary(x, T, H, D, x_stride_t, x_stride_h, pos, table, max_pos, R, offset, interleaved, inverse,
                              dtype, y, y_stride_t, y_stride_h, reinterpret_cast<cudaStream_t>(stream));
}

sgq_status sgq_latent_append(const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k, int64_t k_stride,
                             const void* latent, int64_t latent_stride, const int64_t* pos, const int64_t* slots,
                             const float* table, int64_t max_pos, int64_t T, int64_t H, int64_t L, int R,
                             int interleaved, int dtype, void* q_out, int64_t qo_stride_t, int64_t qo_stride_h,
                             void* k_out, int64_t ko_stride, void* cache, int64_t pages, int64_t page,
                             int64_t cache_stride_page, int64_t cache_stride_row, sgq_stream_t stream) {
    if (T < 0 || T >= (int64_t(1) << 31) || H < 0 || H > 65535 || L <= 0 || L % 8 != 0 || L > 65536 || max_pos <= 0 ||
        !good_rotation(R, interleaved) || R > 256 || !good_dtype(dtype) ||
        !good_strides({q_stride_t, q_stride_h, k_stride, latent_stride, qo_stride_t, qo_stride_h, ko_stride,
                       cache_stride_page, cache_stride_row}))
        return SGQ_ERR_INVALID_ARG;
    if (pages < 0 || page <= 0 || page >= (int64_t(1) << 31) || pages >= (int64_t(1) << 31) ||
        cache_stride_row < L + R || cache_stride_page < 0)
        return SGQ_ERR_INVALID_ARG;
    if (T == 0) return SGQ_OK;
    if (q == q_out && H > 0 && (q_stride_t != qo_stride_t || q_stride_h != qo_stride_h)) return SGQ_ERR_INVALID_ARG;
    if (H > 0 && ((T > 1 && qo_stride_t < R) || (H > 1 && qo_stride_h < R))) return SGQ_ERR_INVALID_ARG;
    if (k_out && T > 1 && ko_stride < R) return SGQ_ERR_INVALID_ARG;
    if (!k || !latent || !pos || !slots || !table || !cache || (H > 0 && (!q || !q_out))) return SGQ_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(q_out) || !aligned16(k) || !aligned16(latent) || !aligned16(table) ||
        !aligned16(k_out) || !aligned16(cache) || !aligned_to(pos, 8) || !aligned_to(slots, 8))
        return SGQ_ERR_MISALIGNED;
    return sgq::launch_latent_append(q, q_stride_t, q_stride_h, k, k_stride, latent, latent_stride, pos, slots, table,
                                     max_pos, T, H, L, R, interleaved, dtype, q_out, qo_stride_t, qo_stride_h, k_out,
                                     ko_stride, cache, pages, page, cache_stride_page, cache_stride_row,
                                     reinterpret_cast<cudaStream_t>(stream));
}

sgq_status sgq_latent_attention_workspace(int64_t T, int64_t H, int64_t L, int64_t* bytes) {
    if (bytes == nullptr || !good_rows(T, H) || L <= 0 || L % 128 != 0 || L > 512) return SGQ_ERR_INVALID_ARG;
    return sgq::latent_attention_workspace(T, H, L, bytes);
}

sgq_status sgq_latent_attention(const void* q, int64_t q_stride_row, int64_t T, int64_t H, const void* cache,
                                int64_t pages, int64_t page, int64_t cache_stride_page, int64_t cache_stride_row,
                                int64_t L, int R, const int32_t* page_table, int64_t table_width, int64_t B,
                                const int32_t* kv_lens, const int32_t* q_starts, float scale, int dtype, void* out,
                                float* lse, void* workspace, int64_t workspace_bytes, sgq_stream_t stream) {
    const bool stall = dtype == (SGQ_BF16 | SGQ_LATENT_TEST_TIMEOUT);
    if (stall) dtype = SGQ_BF16;
    if (!good_rows(T, H) || B < 0 || B >= (int64_t(1) << 31) || L <= 0 || L % 128 != 0 || L > 512 || R < 8 || R > 64 ||
        R % 8 != 0 || !good_dtype(dtype) ||
        !good_strides({q_stride_row, cache_stride_page, cache_stride_row}) || !(std::isfinite(scale) && scale > 0.0f))
        return SGQ_ERR_INVALID_ARG;
    if (pages <= 0 || pages >= (int64_t(1) << 31) || page <= 0 || page % 16 != 0 || page >= (int64_t(1) << 31) ||
        table_width < 0 || table_width >= (int64_t(1) << 31) || table_width * page > (int64_t(1) << 31) - 256 ||
        q_stride_row < L + R || cache_stride_row < L + R || cache_stride_page / page < cache_stride_row)
        return SGQ_ERR_INVALID_ARG;
    if (q_starts == nullptr && T != B) return SGQ_ERR_INVALID_ARG;
    if (T == 0) return SGQ_OK;
    if (B == 0 || !q || !cache || !kv_lens || !out || (table_width > 0 && !page_table) || !workspace)
        return SGQ_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(cache) || !aligned16(out) || !aligned16(workspace) || !aligned_to(page_table, 4) ||
        !aligned_to(kv_lens, 4) || !aligned_to(q_starts, 4) || !aligned_to(lse, 4))
        return SGQ_ERR_MISALIGNED;
    int64_t need = 0;
    sgq_status rc = sgq::latent_attention_workspace(T, H, L, &need);
    if (rc != SGQ_OK) return rc;
    if (workspace_bytes < need) return SGQ_ERR_INVALID_ARG;
    sgq::LatentArgs a{};
    a.q = q; a.cache = cache; a.page_table = page_table; a.kv_lens = kv_lens; a.q_starts = q_starts; a.out = out;
    a.lse = lse; a.workspace = workspace; a.q_row = q_stride_row; a.T = T; a.B = B; a.pages = pages;
    a.c_page = cache_stride_page; a.c_row = cache_stride_row; a.table_width = table_width;
    a.H = static_cast<int>(H); a.L = static_cast<int>(L); a.R = R; a.page = static_cast<int>(page);
    a.dtype = dtype; a.stall = stall;
    a.scale = scale;
    return sgq::launch_latent_attention(a, reinterpret_cast<cudaStream_t>(stream));
}

sgq_status sgq_latent_prefill(const void* q, int64_t q_stride_t, int64_t q_stride_h, int64_t T, const void* k,
                              int64_t k_stride_t, int64_t k_stride_h, const void* k_rot, int64_t kr_stride,
                              const void* v, int64_t v_stride_t, int64_t v_stride_h, int64_t S, int64_t H, int64_t N,
                              int R, const int32_t* q_starts, const int32_t* kv_starts, int64_t B, float scale,
                              int causal, int dtype, void* out, float* lse, sgq_stream_t stream) {
    const bool stall = dtype == (SGQ_BF16 | SGQ_LATENT_TEST_TIMEOUT);
    if (stall) dtype = SGQ_BF16;
    if (T < 0 || S < 0 || B < 0 || H <= 0 || H > 65535 || T >= (int64_t(1) << 31) || S >= (int64_t(1) << 31) ||
        B >= (int64_t(1) << 31) || (N != 64 && N != 128) || R < 8 || R > 64 || R % 8 != 0 || !good_dtype(dtype) ||
        !good_strides({q_stride_t, q_stride_h, k_stride_t, k_stride_h, kr_stride, v_stride_t, v_stride_h}) ||
        (causal != 0 && causal != 1) || !(std::isfinite(scale) && scale > 0.0f))
        return SGQ_ERR_INVALID_ARG;
    // (rows and heads one after the other in memory: no broadcast dimensions)
    if ((T > 1 && q_stride_t == 0) || (S > 1 && (k_stride_t == 0 || v_stride_t == 0 || kr_stride == 0)) ||
        (H > 1 && (q_stride_h == 0 || k_stride_h == 0 || v_stride_h == 0)))
        return SGQ_ERR_INVALID_ARG;
    if (T == 0) return SGQ_OK;
    if (B == 0 || !q || !q_starts || !kv_starts || !out || (S > 0 && (!k || !k_rot || !v))) return SGQ_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(k_rot) || !aligned16(v) || !aligned16(out) ||
        !aligned_to(q_starts, 4) || !aligned_to(kv_starts, 4) || !aligned_to(lse, 4))
        return SGQ_ERR_MISALIGNED;
    sgq::PrefillArgs a{};
    a.q = q; a.k = k; a.k_rot = k_rot; a.v = v; a.q_starts = q_starts; a.kv_starts = kv_starts; a.out = out; a.lse = lse;
    a.q_t = q_stride_t; a.q_h = q_stride_h; a.k_t = k_stride_t; a.k_h = k_stride_h; a.kr_t = kr_stride;
    a.v_t = v_stride_t; a.v_h = v_stride_h; a.T = T; a.S = S; a.B = B;
    a.H = static_cast<int>(H); a.N = static_cast<int>(N); a.R = R; a.causal = causal;
    a.dtype = dtype; a.stall = stall;
    a.scale = scale;
    return sgq::launch_latent_prefill(a, reinterpret_cast<cudaStream_t>(stream));
}

const char* sgq_status_string(sgq_status s) {
    switch (s) {
        case SGQ_OK: return "SGQ_OK";
        case SGQ_ERR_INVALID_ARG: return "SGQ_ERR_INVALID_ARG";
        case SGQ_ERR_UNSUPPORTED: return "SGQ_ERR_UNSUPPORTED";
        case SGQ_ERR_MISALIGNED: return "SGQ_ERR_MISALIGNED";
        case SGQ_ERR_CUDA: return "SGQ_ERR_CUDA";
        case SGQ_ERR_TIMEOUT: return "SGQ_ERR_TIMEOUT";
    }
    return "SGQ_ERR_UNKNOWN";
}

sgq_status sgq_device_status(sgq_stream_t stream) {
    return sgq::read_and_clear_device_status(reinterpret_cast<cudaStream_t>(stream));
}

uint64_t sgq_launch_count(void) { return sgq::g_launches.load(std::memory_order_relaxed); }

uint64_t sgq_allocated_bytes(void) { return sgq::allocated_bytes(); }

sgq_status sgq_gemm_plan(int64_t M, int64_t N, int64_t K, int blk_k, int sm_count, int32_t* out) {
    if (out == nullptr || M < 1 || N < 1 || K < 1 || (blk_k != 32 && blk_k != 128) || sm_count < 1)
        return SGQ_ERR_INVALID_ARG;
    return sgq::gemm_plan_query(M, N, K, blk_k, sm_count, out);
}

sgq_status sgq_gemm_plan_pow2(int64_t M, int64_t N, int64_t K, int blk_k, int sm_count, int e8, int32_t* out) {
    if (out == nullptr || M < 1 || N < 1 || K < 1 || (blk_k != 32 && blk_k != 128) || sm_count < 2 ||
        (e8 != 0 && e8 != 1))
        return SGQ_ERR_INVALID_ARG;
    return sgq::gemm_plan_pow2_query(M, N, K, blk_k, sm_count, e8, out);
}

int sgq_version(void) { return 104; }

}  // extern "C"
