// Internal declarations shared by the translation units of the library.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "compfp32.h"

namespace compfp32 {

// a * b in *out, false if it is negative or overflows.
inline bool mul_ok(int64_t a, int64_t b, int64_t* out)
{
    if (a < 0 || b < 0)
        return false;
    if (a != 0 && b > INT64_MAX / a)
        return false;
    *out = a * b;
    return true;
}

// Byte ranges [a, a+na) and [b, b+nb) overlap.
inline bool overlap(const void* a, int64_t na, const void* b, int64_t nb)
{
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    return na > 0 && nb > 0 && pa < pb + static_cast<uintptr_t>(nb) && pb < pa + static_cast<uintptr_t>(na);
}

// Bytes from the first to the last element of a [tokens, heads, dim] tensor
// with these token and head strides (in elements of `elem` bytes; not negative).
inline bool strided_bytes(int64_t tokens, int64_t heads, int64_t dim, int64_t token, int64_t head, int64_t elem,
                          int64_t* bytes)
{
    int64_t a, b;
    *bytes = 0;
    if (tokens < 0 || heads < 0 || dim < 0 || token < 0 || head < 0)
        return false;
    if (tokens == 0 || heads == 0 || dim == 0)
        return true;
    if (!mul_ok(tokens - 1, token, &a) || !mul_ok(heads - 1, head, &b) || a > INT64_MAX / 64 || b > INT64_MAX / 64)
        return false;
    *bytes = elem * (a + b + dim);
    return true;
}

// Properties of the current device, checked once per device.
struct DeviceInfo {
    int device;
    int sm_count;
};

// COMP_OK and fills `info` if the current device is compute capability 10.3.
comp_status_t current_device(DeviceInfo* info);

// Launchers (arguments already validated; sizes > 0).
comp_status_t launch_split(const float* x, uint16_t* hi, uint16_t* lo, int64_t n, const DeviceInfo& dev,
                           cudaStream_t stream);
// One launch: x [M, K] split into planes [M, Kp] (Kp >= K, a multiple of 8)
// and W [N, K] copied into wp [N, Kp], all zero-padded past K.
comp_status_t launch_prep_padded(const float* x, const uint16_t* W, uint16_t* hi, uint16_t* lo, uint16_t* wp,
                                 int64_t M, int64_t N, int64_t K, int64_t Kp, const DeviceInfo& dev,
                                 cudaStream_t stream);
comp_status_t launch_geglu(const float* gate, const float* up, float* out, int64_t n, const DeviceInfo& dev,
                           cudaStream_t stream);
comp_status_t launch_merge(const float* acc_hi, const float* acc_lo, float* y, int64_t n, const DeviceInfo& dev,
                           cudaStream_t stream);
comp_status_t launch_gemm_simt(const float* x, const uint16_t* W, float* y, int64_t M, int64_t N, int64_t K,
                               const DeviceInfo& dev, cudaStream_t stream);
// Optional FP32 operations on the merged projection in the product kernels'
// epilogue (GEGLU feed-forward step): y = gelu(gate) * (y + bias).
struct Epilogue {
    const float* bias = nullptr;  // [N] (nullptr: none)
    const float* gate = nullptr;  // [M, N] row-major (nullptr: factor 1)
};

// Fused split and swapped-operand product for at most 32 rows of x (K a
// multiple of 8, x and W 16-byte aligned), with K split over a cluster when W
// has few tiles of 128 rows.
bool swap_fused_preferred(const float* x, const uint16_t* W, int64_t M, int64_t N, int64_t K);
// Given a workspace, whether the two-pass form beats the fused swapped kernel
// for a shape that swap_fused_preferred accepts (17 to 32 rows, no split of K).
bool swap_two_pass_better(int64_t M, int64_t N, int64_t K, const DeviceInfo& dev);
comp_status_t launch_swap_fused(const float* x, const uint16_t* W, float* y, int64_t M, int64_t N, int64_t K,
                                const DeviceInfo& dev, cudaStream_t stream, const Epilogue& epi = Epilogue{});
// Fused split and product on CTA pairs (K a multiple of 8, x and W 16-byte
// aligned); preferred for more than 128 rows once the output fills about a
// wave of tiles.
bool fused_pair_preferred(const float* x, const uint16_t* W, int64_t M, int64_t N, int64_t K, const DeviceInfo& dev);
comp_status_t launch_fused_pair(const float* x, const uint16_t* W, float* y, int64_t M, int64_t N, int64_t K,
                                const DeviceInfo& dev, cudaStream_t stream, const Epilogue& epi = Epilogue{});
// variant: 0 automatic, 1 TMA loads, 2 plain loads (both one CTA per tile),
// 3 operands swapped with the split fused (M <= 32), 4 CTA pairs with the
// split fused.
comp_status_t launch_gemm_tc(const float* x, const uint16_t* W, float* y, int64_t M, int64_t N, int64_t K,
                             int variant, const DeviceInfo& dev, cudaStream_t stream, const Epilogue& epi = Epilogue{});

// The two products and the merge from split planes (hi, lo: [M, K] FP16).
// Needs 16-byte aligned hi, lo, W and K % 8 == 0 (else COMP_ERR_INVALID_VALUE).
bool gemm_f16x2_supported(const void* hi, const void* lo, const void* W, int64_t K);
// variant: 0 automatic, 1 one CTA per 128-row tile, 2 CTA pairs on 256-row
// tiles, 3 operands swapped (M <= 32).
// stall: diagnostic run of the CTA-pair (variant 2) or swapped (variant 3)
// kernel whose producer leaves out its first stage's loads (see
// comp_check_stalled_pipeline).
comp_status_t launch_gemm_f16x2(const uint16_t* hi, const uint16_t* lo, const uint16_t* W, float* y, int64_t M,
                                int64_t N, int64_t K, int variant, const DeviceInfo& dev, cudaStream_t stream,
                                const Epilogue& epi = Epilogue{}, bool stall = false);

// Whether a cache descriptor is one that the kernels take; the bytes of its
// k (and of its v).
bool kv_cache_ok(const comp_kv_cache_t* cache, int64_t* bytes);

// Attention of single tokens over a cache (arguments validated; batch > 0), and
// whether its line of tiles can be counted in ints (batch * heads can).
bool attn_decode_countable(const comp_kv_cache_t& cache, int64_t batch, int heads, int64_t width);
int64_t attn_decode_bytes(const comp_kv_cache_t& cache, int64_t batch, int heads, int64_t shared_pages);
comp_status_t launch_attn_decode(const comp_kv_cache_t& cache, const float* q, int64_t q_token, int64_t q_head,
                                 int heads, float scale, const int32_t* table, int64_t batch, int64_t width,
                                 const int32_t* lengths, int64_t shared_pages, float* out, float* lse,
                                 void* workspace, const DeviceInfo& dev, cudaStream_t stream);

// One thread runs a bounded wait that cannot succeed (comp_check_wait_timeout).
comp_status_t launch_check_wait_timeout(cudaStream_t stream);

// Reads and clears the fault word of the tensor-core kernels (after the stream
// has been synchronised).
comp_status_t read_and_clear_fault(cudaStream_t stream, uint32_t* where);
// The same of the attention kernels; `where` is written only if there is a fault.
comp_status_t read_and_clear_attn_fault(cudaStream_t stream, uint32_t* where);
comp_status_t read_and_clear_decode_fault(cudaStream_t stream, uint32_t* where);

// Packed attention (arguments validated; sizes > 0 but total_k) and the
// workspace it needs for k and v.
int64_t attn_stage_bytes(const comp_attn_t& a, int kv_bytes, const void* k, const void* v);
comp_status_t launch_attn(const comp_attn_t& a, const float* q, const void* k, const void* v, int kv_bytes,
                          const int32_t* cu_q, const int32_t* cu_k, float* out, float* lse, void* workspace,
                          const DeviceInfo& dev, cudaStream_t stream);

inline comp_status_t launch_status()
{
    return cudaGetLastError() == cudaSuccess ? COMP_OK : COMP_ERR_LAUNCH;
}

}  // namespace compfp32
