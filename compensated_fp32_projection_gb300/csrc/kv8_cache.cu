// Writing keys and values to a paged cache in 8 bits, and reading them back.
//
// Sixteen tokens of a head on a page are a block, and share a scale:
//   scale = max(kept, rn(max |x| * rn(1/127))), 0 where that is below 2^-126;
//   code  = rint(rn(x * rn(1/scale))), within +-127;       value = code * scale.
// `kept` is the block's scale where tokens before the first new one stay in it;
// their codes become rint(rn(code * rn(kept/scale))).  Every operation is a
// binary32 one, so the codes follow from the inputs bit for bit.  A block grows
// by some tokens at a time; a token's codes are rounded again only when a larger
// one arrives (about three times in 16 tokens of one distribution), and each time
// by half a step of a scale that is smaller than the last.
// An infinity or a NaN takes the code -128, which reads as NaN, and no part in the
// scale; the sign of the block's scale says that it has such codes, so that the
// kernels that read look for them in those blocks only.
//
// Both kernels stream, 5 bytes a value (6 and 3 with keys and values that are read
// back as FP16), and HBM is the bound.  A warp takes a block of a head: its 16
// rows are all loaded before the first is used (up to 64 values a lane, the block
// passes through registers once), and the maximum is one reduction in the warp.
#include <cuda_fp16.h>

#include <cmath>

#include "internal.h"
#include "ptx.cuh"
#include "rope.cuh"
#include "tc_util.cuh"

namespace compfp32 {
namespace {

constexpr int kBlock = COMP_KV8_BLOCK;
constexpr int kThreads = 256;
constexpr uint32_t kNan4 = 0x80808080u;  // four codes of -128

struct Params {
    comp_kv8_cache_t cache;
    const int32_t* table;
    const int32_t* cu;      // nullptr: one token for each row
    const int32_t* start;
    int64_t rows, width, total;
    int64_t slots;          // see slot_of_row
};

// Blocks are numbered without a sum over the rows: row r's begin at
// cu[r] / 16 + 2 r, which leaves room for every block that its tokens can touch
// (n tokens from anywhere in a block touch at most n / 16 + 2).
__device__ __forceinline__ int64_t first_token(const Params& p, int64_t row)
{
    const int64_t n = p.cu[row];
    return n < 0 ? 0 : (n > p.total ? p.total : n);
}

__device__ __forceinline__ int64_t slot_of_row(const Params& p, int64_t row)
{
    return first_token(p, row) / kBlock + 2 * row;
}

// A block of a row: tokens `from` to `to` of its 16 are packed tokens token0 + from, ...
struct Work {
    int64_t row, token0, position;  // position of the block's first token
    int from, to;
    bool begins;                    // the row's first block
};

// By a whole warp: the last row that begins at or before this slot, 32 at a time.
__device__ __forceinline__ Work work_of(const Params& p, int64_t slot)
{
    Work w{0, 0, 0, 0, 0, false};
    int64_t t0, t1, nth;
    if (!p.cu) {
        w.row = t0 = slot;
        t1 = t0 + 1;
        nth = 0;
    } else {
        const int lane = threadIdx.x & 31;
        int64_t lo = 0, n = p.rows + 1;  // row p.rows: the tokens behind the last sequence
        while (n > 1) {
            const int64_t step = (n + 31) / 32, r = lo + lane * step;
            const unsigned in = __ballot_sync(0xffffffffu, r < lo + n && slot_of_row(p, r) <= slot);
            const int last = in ? 31 - __clz(in) : 0;
            n = n - last * step < step ? n - last * step : step;
            lo += last * step;
        }
        w.row = lo;
        t0 = first_token(p, lo);
        t1 = lo < p.rows ? first_token(p, lo + 1) : p.total;
        nth = slot - slot_of_row(p, lo);
    }
    if (nth < 0 || t1 < t0)  // only where cu does not ascend from 0
        return w;
    const int64_t start = w.row < p.rows ? p.start[w.row] : 0;
    const int lead = static_cast<int>(start & (kBlock - 1));
    const int64_t before = nth * kBlock - lead, rest = t1 - t0 - before;  // the row's tokens before this block, and from it on
    w.position = start + before;
    w.token0 = t0 + before;
    w.from = nth == 0 ? lead : 0;
    w.to = rest > kBlock ? kBlock : (rest < 0 ? 0 : static_cast<int>(rest));
    w.begins = nth == 0;
    return w;
}

// The page that has a position, or -1.
__device__ __forceinline__ int64_t page_of(const Params& p, const Work& w)
{
    const int64_t col = w.position < 0 || w.row >= p.rows ? p.width : w.position / p.cache.page_size;
    const int64_t page = col < p.width ? p.table[w.row * p.width + col] : -1;
    return page < p.cache.pages ? page : -1;
}

// How a warp goes over a block: lanes_a_row lanes have a row's codes, four each.
struct Lanes {
    int rows_at_once, row, d;
    bool in;
    __device__ __forceinline__ explicit Lanes(int dim)
    {
        const int lane = threadIdx.x & 31, a_row = dim / 4;
        rows_at_once = 32 / a_row;
        row = lane / a_row;
        d = lane % a_row * 4;
        in = row < rows_at_once;
    }
};

__device__ __forceinline__ int code_of(float x, float inverse)
{
    if (!(fabsf(x) < INFINITY))
        return -128;
    return static_cast<int>(fminf(fmaxf(rintf(__fmul_rn(x, inverse)), -127.0f), 127.0f));
}

struct Source {
    const float* x;
    int64_t token, head;
    int vec;
};

// STEPS: how often the warp moves on in a block's 16 rows, 16 for heads wider
// than 64 and 8 for others.
template <int STEPS>
__global__ void __launch_bounds__(kThreads) append8_kernel(const Params p, const Source k, const Source v,
                                                           const comp_rope_t rope, const int wide)
{
    grid_dependency_launch();
    const comp_kv8_cache_t& c = p.cache;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    const int heads = 2 * c.kv_heads, blocks = c.page_size / kBlock;
    const Lanes at(c.head_dim);
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); u < p.slots * heads;
         u += warps) {
        const Work w = work_of(p, u / heads);
        const int64_t page = w.row < p.rows && w.to > w.from ? page_of(p, w) : -1;
        if (page < 0)
            continue;
        const int head = static_cast<int>(u % heads) / 2, is_v = static_cast<int>(u % 2);
        const Source& src = is_v ? v : k;
        const bool turns = !is_v && rope.rot > 0;
        const int slot = static_cast<int>(w.position % c.page_size);
        const int64_t unit = page * c.kv_heads + head;
        int8_t* const codes = (is_v ? c.v : c.k) + (unit * c.page_size + slot) * c.head_dim;
        float* const scale_at = (is_v ? c.v_scale : c.k_scale) + unit * blocks + slot / kBlock;
        const float* const x0 = src.x + w.token0 * src.token + head * src.head;
        const float was = w.begins && w.from > 0 ? *scale_at : 0.0f;
        float4 x[STEPS];
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            const int t = i * at.rows_at_once + at.row;
            x[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (!at.in || t < w.from || t >= w.to)
                continue;
            const float* const row = x0 + t * src.token;
            if (turns)
                x[i] = load_rotated(row, at.d, rope, angles_of(rope, w.position + t), src.vec != 0,
                                    wide != 0);
            else if (src.vec)
                x[i] = __ldcs(reinterpret_cast<const float4*>(row + at.d));
            else
                x[i] = make_float4(row[at.d], row[at.d + 1], row[at.d + 2], row[at.d + 3]);
        }
        // the largest finite magnitude; as bits they have the same order
        float top = 0.0f;
        bool odd = false;
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            const float m[4] = {fabsf(x[i].x), fabsf(x[i].y), fabsf(x[i].z), fabsf(x[i].w)};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool finite = m[e] < INFINITY;
                odd |= !finite;
                top = finite ? fmaxf(top, m[e]) : top;
            }
        }
        top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
        odd = __any_sync(0xffffffffu, odd) || (__float_as_uint(was) >> 31) != 0;
        const float kept = fabsf(was);
        float scale = __fmul_rn(top, 0x1.020408p-7f);  // 1/127
        scale = scale < 0x1p-126f ? 0.0f : scale;
        scale = kept > scale ? kept : scale;
        const float inverse = scale > 0.0f ? __frcp_rn(scale) : 0.0f;
        const bool again = kept != scale && w.begins && w.from > 0;
        const float ratio = again && scale > 0.0f ? __fdiv_rn(kept, scale) : 0.0f;
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            const int t = i * at.rows_at_once + at.row;
            if (!at.in || t >= w.to || (t < w.from && !again))
                continue;
            char4* const to = reinterpret_cast<char4*>(codes + static_cast<int64_t>(t) * c.head_dim + at.d);
            int q[4];
            if (t < w.from) {
                const char4 old = *to;
                const int o[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    q[e] = o[e] == -128 ? -128 : static_cast<int>(rintf(__fmul_rn(static_cast<float>(o[e]), ratio)));
            } else {
                q[0] = code_of(x[i].x, inverse);
                q[1] = code_of(x[i].y, inverse);
                q[2] = code_of(x[i].z, inverse);
                q[3] = code_of(x[i].w, inverse);
            }
            *to = make_char4(static_cast<signed char>(q[0]), static_cast<signed char>(q[1]),
                             static_cast<signed char>(q[2]), static_cast<signed char>(q[3]));
        }
        if ((threadIdx.x & 31) == 0)
            *scale_at = odd ? -scale : scale;
    }
}

struct Sink {
    void* x;
    int64_t token, head;
    int vec;
};

__device__ __forceinline__ float value_of(int code, float scale)
{
    return code == -128 ? __int_as_float(0x7fffffff) : __fmul_rn(static_cast<float>(code), scale);
}

template <typename T, int STEPS>
__global__ void __launch_bounds__(kThreads) read8_kernel(const Params p, const Sink k, const Sink v)
{
    grid_dependency_launch();
    const comp_kv8_cache_t& c = p.cache;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    const int heads = 2 * c.kv_heads, blocks = c.page_size / kBlock;
    const Lanes at(c.head_dim);
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); u < p.slots * heads;
         u += warps) {
        const Work w = work_of(p, u / heads);
        if (w.to <= w.from)
            continue;
        const int64_t page = page_of(p, w);  // -1 for tokens of no sequence too: zeros
        const int head = static_cast<int>(u % heads) / 2, is_v = static_cast<int>(u % 2);
        const Sink& dst = is_v ? v : k;
        const int slot = page < 0 ? 0 : static_cast<int>(w.position % c.page_size);
        const int64_t unit = page < 0 ? 0 : page * c.kv_heads + head;
        const int8_t* const codes = (is_v ? c.v : c.k) + (unit * c.page_size + slot) * c.head_dim;
        const float scale = page < 0 ? 0.0f : fabsf((is_v ? c.v_scale : c.k_scale)[unit * blocks + slot / kBlock]);
        char4 q[STEPS];
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            const int t = i * at.rows_at_once + at.row;
            q[i] = make_char4(0, 0, 0, 0);
            if (at.in && t >= w.from && t < w.to && page >= 0)
                q[i] = __ldcs(reinterpret_cast<const char4*>(codes + static_cast<int64_t>(t) * c.head_dim + at.d));
        }
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            const int t = i * at.rows_at_once + at.row;
            if (!at.in || t < w.from || t >= w.to)
                continue;
            T* const to = static_cast<T*>(dst.x) + (w.token0 + t) * dst.token + head * dst.head + at.d;
            const float x[4] = {value_of(q[i].x, scale), value_of(q[i].y, scale), value_of(q[i].z, scale),
                                value_of(q[i].w, scale)};
            if constexpr (sizeof(T) == 4) {
                if (dst.vec) {
                    *reinterpret_cast<float4*>(to) = make_float4(x[0], x[1], x[2], x[3]);
                    continue;
                }
            } else {
                if (dst.vec) {
                    *reinterpret_cast<uint2*>(to) = make_uint2(pack_h2(__floats2half2_rn(x[0], x[1])),
                                                               pack_h2(__floats2half2_rn(x[2], x[3])));
                    continue;
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if constexpr (sizeof(T) == 4)
                    to[e] = x[e];
                else
                    to[e] = __float2half_rn(x[e]);
        }
    }
}

unsigned grid_of(int64_t warps, const DeviceInfo& dev)
{
    const int64_t most = static_cast<int64_t>(dev.sm_count) * 8, g = (warps + kThreads / 32 - 1) / (kThreads / 32);
    return static_cast<unsigned>(g < 1 ? 1 : (g > most ? most : g));
}

// Rows of `elem`-byte values whose parts of four are aligned to their size.
int rows_vec(const void* x, int64_t token, int64_t head, int elem)
{
    return reinterpret_cast<uintptr_t>(x) % (4 * static_cast<uintptr_t>(elem)) == 0 && token % 4 == 0 && head % 4 == 0;
}

// The slots of a call; see slot_of_row.  One more for the tokens behind the last sequence.
int64_t slots_of(int64_t total, int64_t rows, const int32_t* cu)
{
    return cu ? total / kBlock + 2 * rows + 1 : rows;
}

bool apart(const void* out, int64_t bytes, const void* const (&p)[8], const int64_t (&n)[8])
{
    for (int i = 0; i < 8; ++i)
        if (overlap(out, bytes, p[i], n[i]))
            return false;
    return true;
}

comp_status_t read8(const comp_kv8_cache_t* cache, void* k, void* v, int elem, int64_t k_token, int64_t k_head,
                    int64_t v_token, int64_t v_head, int64_t total, const int32_t* table, int64_t rows, int64_t width,
                    const int32_t* cu, const int32_t* start, comp_stream_t stream)
{
    int64_t bytes, scales, entries, kb, vb;
    if (!kv8_cache_ok(cache, &bytes, &scales) ||
        !kv_table_ok(cache->pages, cache->page_size, rows, width, &entries) || total < 0 || total > INT32_MAX ||
        (!cu && total != rows) ||
        !strided_bytes(total, cache->kv_heads, cache->head_dim, k_token, k_head, elem, &kb) ||
        !strided_bytes(total, cache->kv_heads, cache->head_dim, v_token, v_head, elem, &vb) ||
        !rows_apart(total, cache->kv_heads, cache->head_dim, k_token, k_head) ||
        !rows_apart(total, cache->kv_heads, cache->head_dim, v_token, v_head))
        return COMP_ERR_INVALID_VALUE;
    if (total == 0)
        return COMP_OK;
    const int64_t eb = 4 * entries, cb = cu ? 4 * (rows + 1) : 0, sb = 4 * rows;
    if (!k || !v || (eb > 0 && !table) || (sb > 0 && !start) || overlap(k, kb, v, vb))
        return COMP_ERR_INVALID_VALUE;
    const void* const in[8] = {cache->k, cache->v, cache->k_scale, cache->v_scale, table, cu, start, nullptr};
    const int64_t n[8] = {bytes, bytes, scales, scales, eb, cb, sb, 0};
    if (!apart(k, kb, in, n) || !apart(v, vb, in, n))
        return COMP_ERR_INVALID_VALUE;
    DeviceInfo dev;
    const comp_status_t st = current_device(&dev);
    if (st != COMP_OK)
        return st;
    const Params p{*cache, table, cu, start, rows, width, total, slots_of(total, rows, cu)};
    const Sink ks{k, k_token, k_head, rows_vec(k, k_token, k_head, elem)};
    const Sink vs{v, v_token, v_head, rows_vec(v, v_token, v_head, elem)};
    const unsigned grid = grid_of(p.slots * 2 * cache->kv_heads, dev);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (elem == 4) {
        if (cache->head_dim > 64)
            read8_kernel<float, 16><<<grid, kThreads, 0, s>>>(p, ks, vs);
        else
            read8_kernel<float, 8><<<grid, kThreads, 0, s>>>(p, ks, vs);
    } else {
        if (cache->head_dim > 64)
            read8_kernel<__half, 16><<<grid, kThreads, 0, s>>>(p, ks, vs);
        else
            read8_kernel<__half, 8><<<grid, kThreads, 0, s>>>(p, ks, vs);
    }
    return launch_status();
}

}  // namespace

bool kv8_cache_ok(const comp_kv8_cache_t* c, int64_t* bytes, int64_t* scales)
{
    if (!c || c->pages < 0 || c->pages > INT32_MAX / 2 || c->kv_heads <= 0 || c->kv_heads > 65535 ||
        c->head_dim <= 0 || c->head_dim > 128 || c->head_dim % 16 != 0)
        return false;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
        return false;
    const int64_t page = static_cast<int64_t>(c->kv_heads) * c->page_size * c->head_dim;
    if (!mul_ok(c->pages, page, bytes) || *bytes > INT64_MAX / 4)
        return false;
    *scales = c->pages * c->kv_heads * (c->page_size / kBlock) * 4;
    if (*bytes == 0)
        return true;
    const void* const p[] = {c->k, c->v, c->k_scale, c->v_scale};
    const int64_t n[] = {*bytes, *bytes, *scales, *scales};
    for (int i = 0; i < 4; ++i) {
        if (!p[i] || (reinterpret_cast<uintptr_t>(p[i]) & (i < 2 ? 15u : 3u)) != 0)
            return false;
        for (int j = 0; j < i; ++j)
            if (overlap(p[i], n[i], p[j], n[j]))
                return false;
    }
    return true;
}

}  // namespace compfp32

using namespace compfp32;

extern "C" {

comp_status_t comp_kv8_append_f32(const comp_kv8_cache_t* cache, const float* k, const float* v, int64_t k_token,
                                  int64_t k_head, int64_t v_token, int64_t v_head, int64_t total,
                                  const int32_t* table, int64_t rows, int64_t width, const int32_t* cu,
                                  const int32_t* start, const comp_rope_t* rope, comp_stream_t stream)
{
    int64_t bytes, scales, entries, kb, vb, rb;
    if (!kv8_cache_ok(cache, &bytes, &scales) ||
        !kv_table_ok(cache->pages, cache->page_size, rows, width, &entries) || total < 0 || total > INT32_MAX ||
        (!cu && total != rows) ||
        !strided_bytes(total, cache->kv_heads, cache->head_dim, k_token, k_head, 4, &kb) ||
        !strided_bytes(total, cache->kv_heads, cache->head_dim, v_token, v_head, 4, &vb) ||
        !rope_ok(rope, cache->head_dim, &rb))
        return COMP_ERR_INVALID_VALUE;
    if (total == 0 || bytes == 0 || entries == 0)
        return COMP_OK;
    if (!k || !v || !table || !start)
        return COMP_ERR_INVALID_VALUE;
    const void* const in[8] = {k, v, table, cu, start, rope ? rope->table : nullptr, nullptr, nullptr};
    const int64_t n[8] = {kb, vb, 4 * entries, cu ? 4 * (rows + 1) : 0, 4 * rows, rb, 0, 0};
    if (!apart(cache->k, bytes, in, n) || !apart(cache->v, bytes, in, n) || !apart(cache->k_scale, scales, in, n) ||
        !apart(cache->v_scale, scales, in, n))
        return COMP_ERR_INVALID_VALUE;
    DeviceInfo dev;
    const comp_status_t st = current_device(&dev);
    if (st != COMP_OK)
        return st;
    const Params p{*cache, table, cu, start, rows, width, total, slots_of(total, rows, cu)};
    const Source ks{k, k_token, k_head, rows_vec(k, k_token, k_head, 4)};
    const Source vs{v, v_token, v_head, rows_vec(v, v_token, v_head, 4)};
    const comp_rope_t r = rope ? *rope : comp_rope_t{};
    const int wide = angles_wide(r);
    const unsigned grid = grid_of(p.slots * 2 * cache->kv_heads, dev);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cache->head_dim > 64)
        append8_kernel<16><<<grid, kThreads, 0, s>>>(p, ks, vs, r, wide);
    else
        append8_kernel<8><<<grid, kThreads, 0, s>>>(p, ks, vs, r, wide);
    return launch_status();
}

comp_status_t comp_kv8_read_f32(const comp_kv8_cache_t* cache, float* k, float* v, int64_t k_token, int64_t k_head,
                                int64_t v_token, int64_t v_head, int64_t total, const int32_t* table, int64_t rows,
                                int64_t width, const int32_t* cu, const int32_t* start, comp_stream_t stream)
{
    return read8(cache, k, v, 4, k_token, k_head, v_token, v_head, total, table, rows, width, cu, start, stream);
}

comp_status_t comp_kv8_read_f16(const comp_kv8_cache_t* cache, uint16_t* k, uint16_t* v, int64_t k_token,
                                int64_t k_head, int64_t v_token, int64_t v_head, int64_t total, const int32_t* table,
                                int64_t rows, int64_t width, const int32_t* cu, const int32_t* start,
                                comp_stream_t stream)
{
    return read8(cache, k, v, 2, k_token, k_head, v_token, v_head, total, table, rows, width, cu, start, stream);
}

}  // extern "C"
