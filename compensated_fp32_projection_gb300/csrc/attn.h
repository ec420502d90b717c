// What the attention kernels share: the softmax's constants and arithmetic,
// bounded waits, and tensor maps over pages.
#pragma once

#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"
#include "tc_util.cuh"

namespace compfp32 {

constexpr float kAttnLog2E = 1.4426950408889634f;
constexpr float kAttnLn2 = 0.6931471805599453f;
constexpr float kAttnPScale = 16384.0f;             // 2^14: see split_p
constexpr float kAttnLargeScore = 1048576.0f;       // 2^20: from here on s c - m is rounded step by step
constexpr long long kAttnWaitLimit = 1ll << 31;     // cycles (about a second)

// The fault word of the including file's kernels.
static __device__ uint32_t g_attn_fault_word;

__device__ __forceinline__ bool attn_wait(uint64_t* bar, uint32_t parity, int* abort_flag, uint32_t code)
{
    if (mbar_try_wait(bar, parity))
        return true;
    const long long start = clock64();
    while (true) {
        if (mbar_try_wait_sleep(bar, parity, 20000))
            return true;
        if (*reinterpret_cast<volatile int*>(abort_flag))
            return false;
        if (clock64() - start > kAttnWaitLimit) {
            atomicCAS(&g_attn_fault_word, 0u, code);
            *reinterpret_cast<volatile int*>(abort_flag) = 1;
            return false;
        }
    }
}

// The same for a barrier that the other CTA of a cluster arrives on too.
__device__ __forceinline__ bool attn_wait_cluster(uint64_t* bar, uint32_t parity, int* abort_flag, uint32_t code)
{
    const long long start = clock64();
    while (!mbar_try_wait_acquire_cluster(bar, parity)) {
        if (*reinterpret_cast<volatile int*>(abort_flag))
            return false;
        if (clock64() - start > kAttnWaitLimit) {
            atomicCAS(&g_attn_fault_word, 0u, code);
            *reinterpret_cast<volatile int*>(abort_flag) = 1;
            return false;
        }
    }
    return true;
}

// Warp-wide: lane 0 waits, and on success every lane observes the phase itself.
__device__ __forceinline__ bool attn_warp_wait(uint64_t* bar, uint32_t parity, int* abort_flag, uint32_t code)
{
    bool ok = true;
    if ((threadIdx.x & 31) == 0)
        ok = attn_wait(bar, parity, abort_flag, code);
    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
    if (ok)
        (void)mbar_try_wait(bar, parity);
    return ok;
}

// Lane 0 waits for the warp; for loads from tensor memory, which
// tcgen05.fence::after_thread_sync orders after this.
__device__ __forceinline__ bool attn_lane0_wait(uint64_t* bar, uint32_t parity, int* abort_flag, uint32_t code)
{
    bool ok = true;
    if ((threadIdx.x & 31) == 0)
        ok = attn_wait(bar, parity, abort_flag, code);
    return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
}

// Wait for what was issued before the CTA exits after an abort.
__device__ __forceinline__ void attn_drain_wait(uint64_t* bar, uint32_t parity)
{
    const long long start = clock64();
    while (!mbar_try_wait(bar, parity) && clock64() - start < kAttnWaitLimit) {
    }
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two FP32 operations at once, each rounded to nearest even.
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ uint64_t u2_bits(uint32_t a, uint32_t b)
{
    return static_cast<uint64_t>(a) | (static_cast<uint64_t>(b) << 32);
}

// Two weights, 2^14 p each with 0 <= p <= 1, as FP16 pairs hi and lo with
// hi + lo = 2^14 p: lo = fp16(2^14 p - hi), unscaled.  hi is at most 16384 and
// lo has FP16's subnormals down to 2^-24, so what is lost of a weight is at
// most 2^-22 of it or 2^-39 of the largest possible one.
// p - hi is exact, and one operation on the packed hi (an FP16 factor of -1).
__device__ __forceinline__ void split_p(float p0, float p1, uint32_t& hi, uint32_t& lo)
{
    hi = pack_h2(__floats2half2_rn(p0, p1));
    float r0, r1;
    asm("{\n\t.reg .b16 a, b, m;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "mov.b16 m, 0xbc00;\n\t"
        "fma.rn.f32.f16 %0, a, m, %3;\n\t"
        "fma.rn.f32.f16 %1, b, m, %4;\n\t}"
        : "=f"(r0), "=f"(r1)
        : "r"(hi), "f"(p0), "f"(p1));
    lo = pack_h2(__floats2half2_rn(r0, r1));
}

// FP16 [heads][rows][dim] as boxes of box_rows x 64 values, 128-byte swizzled.
// A dimension of extent 1 may have any stride.
inline bool encode_rows(CUtensorMap* map, const void* base, int64_t dim, int64_t rows, int64_t heads,
                        int64_t row_stride, int64_t head_stride, int box_rows)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn)
        return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(heads)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(rows > 1 ? row_stride * 2 : 256),
                                   static_cast<cuuint64_t>(heads > 1 ? head_stride * 2 : 256)};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A cache's k or v: rows are the tokens of one head on one page.
inline bool encode_pages(CUtensorMap* map, const uint16_t* base, const comp_kv_cache_t& c, int box_rows)
{
    return encode_rows(map, base, c.head_dim, c.page_size, c.pages * c.kv_heads, c.head_dim,
                       static_cast<int64_t>(c.page_size) * c.head_dim, box_rows);
}

// Reads and clears a fault word; `where` is written only if it is set.
inline comp_status_t read_and_clear_word(const void* symbol, cudaStream_t stream, uint32_t* where)
{
    uint32_t word = 0;
    const uint32_t zero = 0;
    if (cudaMemcpyFromSymbolAsync(&word, symbol, sizeof(word), 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
        cudaMemcpyToSymbolAsync(symbol, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream) != cudaSuccess ||
        cudaStreamSynchronize(stream) != cudaSuccess) {
        (void)cudaGetLastError();
        return COMP_ERR_CUDA;
    }
    if (word != 0 && where)
        *where = word;
    return word == 0 ? COMP_OK : COMP_ERR_TIMEOUT;
}

// The shared pages of a batch (the first entries of table row 0), in `splits`
// parts, two a CTA if `fold` (an even number of them, up to 128 rows, heads of up
// to 64): out [splits][batch * heads][head_dim], lse [splits][batch * heads].
comp_status_t launch_attn_prefix(const comp_kv_cache_t& cache, const float* q, int64_t q_token, int64_t q_head,
                                 int heads, float scale, const int32_t* table, int64_t batch, const int32_t* lengths,
                                 int64_t shared, int splits, bool fold, float* out, float* lse, const DeviceInfo& dev,
                                 cudaStream_t stream);

}  // namespace compfp32
