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
// Both kernels stream, 5 bytes a value (3 where values are read back as FP16), and
// HBM is the bound.  A warp takes a block of a head: its 16 rows are all loaded
// before the first is used (up to 64 values a lane, the block passes through
// registers once), and the maximum is one reduction in the warp.  Where a block's
// tokens and its page are takes some dependent loads, and its positions' angles are
// the same for all heads: a CTA finds them once for a few blocks (a warp each) and
// then goes over their heads.  With a search by each warp for its block of a head,
// 32768 tokens of 8 heads of 128 took 287 us to write and read back.  They are written in
// 56 us now, 6.0 TB/s, and read in 56.  Where a call raises the scale of a block, its old
// codes take one more round through memory: the last token of each of 64 blocks, 8 heads
// of 128, takes 4.8 us where no scale grows and 11.3 where all do.
#include <cuda_fp16.h>

#include <cmath>
#include <type_traits>

#include "attn.h"
#include "internal.h"
#include "ptx.cuh"
#include "rope.cuh"
#include "tc_util.cuh"

namespace compfp32 {
namespace {

constexpr int kBlock = COMP_KV8_BLOCK;
constexpr int kThreads = 256;

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
    // the row's tokens before this block, and from it on
    const int64_t before = nth * kBlock - lead, rest = t1 - t0 - before;
    w.position = start + before;
    w.token0 = t0 + before;
    w.from = nth == 0 ? lead : 0;
    w.to = rest > kBlock ? kBlock : (rest < 0 ? 0 : static_cast<int>(rest));
    w.begins = nth == 0;
    return w;
}

// The page that has a position, or a negative number.
__device__ __forceinline__ int64_t page_of(const Params& p, int64_t row, int64_t position)
{
    const int64_t col = position < 0 || row >= p.rows ? p.width : position / p.cache.page_size;
    const int64_t page = col < p.width ? p.table[row * p.width + col] : -1;
    return page < p.cache.pages ? page : -1;
}

// Blocks that a CTA finds at once.
constexpr int kMostItems = 4;

struct Item {
    int64_t row, token0, position, unit;  // unit: of the page's first head; negative: no page
    int from, to, slot;
    bool begins;
};

// By all threads: the CTA's blocks, but for their pages; `count` of them are there.
__device__ __forceinline__ int find_items(const Params& p, int items, Item* item)
{
    const int64_t first = static_cast<int64_t>(blockIdx.x) * items;
    const int warp = threadIdx.x >> 5;
    const int count = static_cast<int>(min(static_cast<int64_t>(items), p.slots - first));
    if (warp < count) {
        const Work w = work_of(p, first + warp);
        if ((threadIdx.x & 31) == 0)
            item[warp] = Item{w.row, w.token0, w.position, -1, w.from, w.to, 0, w.begins};
    }
    __syncthreads();
    return count;
}

// Then their pages, for the threads that a later __syncthreads orders behind this.
__device__ __forceinline__ void find_pages(const Params& p, int count, Item* item)
{
    if (threadIdx.x < count) {
        Item& w = item[threadIdx.x];
        const int64_t page = w.to > w.from ? page_of(p, w.row, w.position) : -1;
        w.unit = page < 0 ? -1 : page * p.cache.kv_heads;
        w.slot = page < 0 ? 0 : static_cast<int>(w.position % p.cache.page_size);
    }
}

// How a warp goes over a block: `a_row` lanes have a row, `values` each.
struct Lanes {
    int rows_at_once, row, d;
    bool in;
    __device__ __forceinline__ Lanes(int dim, int values)
    {
        const int lane = threadIdx.x & 31, a_row = dim / values;
        rows_at_once = 32 / a_row;
        row = lane / a_row;
        d = lane % a_row * values;
        in = row < rows_at_once;
    }
};

// rint(rn(x * inverse)) as the low byte of the result, two values: 1.5 2^23 added rounds
// to a whole number, to nearest even.  (The conversion instructions run at a quarter of
// that rate and bounded the kernel.)  No value leaves +-127: inverse is within 2^-23 of
// 127 over the block's largest, or of 1 over a larger scale.
__device__ __forceinline__ uint64_t codes_of(float x, float y, float inverse)
{
    // two products one by one: the compiler fuses a packed one with the addition
    return add2(f2_bits(__fmul_rn(x, inverse), __fmul_rn(y, inverse)), f2_bits(12582912.0f, 12582912.0f));
}

// Four values' codes.
__device__ __forceinline__ uint32_t codes_of(const float4& x, float inverse)
{
    const uint64_t a = codes_of(x.x, x.y, inverse), b = codes_of(x.z, x.w, inverse);
    return __byte_perm(__byte_perm(static_cast<uint32_t>(a), static_cast<uint32_t>(a >> 32), 0x0040),
                       __byte_perm(static_cast<uint32_t>(b), static_cast<uint32_t>(b >> 32), 0x0040), 0x5410);
}

// The largest magnitude of three; NaN if one of them is.
__device__ __forceinline__ float largest(float a, float b, float c)
{
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Four codes as numbers: 2^23 + 128 + code by its bits.
__device__ __forceinline__ float4 numbers_of(uint32_t w, float scale)
{
    const uint32_t u = w ^ 0x80808080u, base = 0x4b000000u;
    const uint64_t bias = f2_bits(-8388736.0f, -8388736.0f), s = f2_bits(scale, scale);
    const uint64_t a = mul2(add2(u2_bits(__byte_perm(u, base, 0x7650), __byte_perm(u, base, 0x7651)), bias), s);
    const uint64_t b = mul2(add2(u2_bits(__byte_perm(u, base, 0x7652), __byte_perm(u, base, 0x7653)), bias), s);
    return make_float4(lo_f(a), hi_f(a), lo_f(b), hi_f(b));
}

// All bits of the bytes of w that are -128, the code of what is no number.
__device__ __forceinline__ uint32_t odd_bytes(uint32_t w)
{
    return __vcmpeq4(w, 0x80808080u);
}

struct Source {
    const float* x;
    int64_t token, head;
    int vec;
};

// How keys turn: not at all; pairs side by side, or halves whose partner of four
// values is four values of another lane; other halves, whose partners are loaded.
enum Turn { kStill, kPairs, kHalves, kOddHalves };

// STEPS: how often the warp moves on in a block's 16 rows, 16 for heads wider
// than 64 and 8 for others.
template <int STEPS, int TURN>
__global__ void __launch_bounds__(kThreads, 2) append8_kernel(const Params p, const Source k, const Source v,
                                                              const comp_rope_t rope, const int items)
{
    grid_dependency_launch();
    __shared__ Item item[kMostItems];
    extern __shared__ __align__(16) float2 angles[];  // [items][kBlock][rot / 2], read two at a time
    const comp_kv8_cache_t& c = p.cache;
    const int heads = 2 * c.kv_heads, blocks = c.page_size / kBlock, half = rope.rot / 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int count = find_items(p, items, item);
    const Lanes at(c.head_dim, 4);
    float4 x[STEPS];
    const int units = count * heads;
    // All 16 rows are new, in places that vector loads take, and the steps fit them.
    auto whole_of = [&](const Item& w, const Source& src) {
        return w.from == 0 && w.to == kBlock && src.vec && STEPS * at.rows_at_once == kBlock;
    };
    // A few new rows, as where each sequence goes on by a token, take one step from the
    // first of them on: a small part of the code, whose fetch is most of such a call.
    auto few_of = [&](const Item& w) { return w.to - w.from <= at.rows_at_once; };
    auto load = [&](int u, auto steps) {
        constexpr int N = decltype(steps)::value;
        const Item& w = item[u / heads];
        const Source& src = u % 2 ? v : k;
        const int t0 = (N == 1 ? w.from : 0) + at.row;
        const float* row = src.x + (w.token0 + t0) * src.token + (u % heads / 2) * src.head + at.d;
        const int64_t step = at.rows_at_once * src.token;
        if (N > 1 && whole_of(w, src)) {
#pragma unroll
            for (int i = 0; i < N; ++i, row += step)
                x[i] = at.in ? __ldcs(reinterpret_cast<const float4*>(row)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i, row += step) {
                const int t = t0 + i * at.rows_at_once;
                x[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (!at.in || t < w.from || t >= w.to)
                    continue;
                if (src.vec)
                    x[i] = __ldcs(reinterpret_cast<const float4*>(row));
                else
                    x[i] = make_float4(row[0], row[1], row[2], row[3]);
            }
        }
    };
    auto write = [&](int u, auto steps) {
        constexpr int N = decltype(steps)::value;
        const Item& w = item[u / heads];
        const int head = u % heads / 2, is_v = u % 2, t0 = (N == 1 ? w.from : 0) + at.row;
        const Source& src = is_v ? v : k;
        const int64_t unit = w.unit + head;
        int8_t* const codes = (is_v ? c.v : c.k) + (unit * c.page_size + w.slot) * c.head_dim + at.d;
        float* const scale_at = (is_v ? c.v_scale : c.k_scale) + unit * blocks + w.slot / kBlock;
        const bool stays = w.begins && w.from > 0;
        const float was = stays ? *scale_at : 0.0f;
        if (TURN != kStill && !is_v) {
            const float2* const turns = angles + u / heads * kBlock * half;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int t = t0 + i * at.rows_at_once;
                const bool here = at.in && t >= w.from && t < w.to && at.d < rope.rot;
                float y[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                if constexpr (TURN == kPairs) {
                    if (here)
#pragma unroll
                        for (int e = 0; e < 4; e += 2)
                            if (at.d + e < rope.rot) {
                                const float2 cs = turns[t * half + (at.d + e) / 2];
                                const float a = y[e], b = y[e + 1];
                                y[e] = turn(a, cs.x, b, cs.y, false);
                                y[e + 1] = turn(b, cs.x, a, cs.y, true);
                            }
                } else if constexpr (TURN == kHalves) {
                    const bool second = at.d >= half;
                    const int partner = (lane + (second ? -half / 4 : half / 4)) & 31, j = second ? at.d - half : at.d;
                    float z[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        z[e] = __shfl_sync(0xffffffffu, y[e], partner);
                    if (here)
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            const float4 cs = *reinterpret_cast<const float4*>(turns + t * half + j + e);
                            y[e] = turn(y[e], cs.x, z[e], cs.y, second);
                            y[e + 1] = turn(y[e + 1], cs.z, z[e + 1], cs.w, second);
                        }
                } else {
                    const float* const row = src.x + (w.token0 + t) * src.token + head * src.head;
                    if (here)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (at.d + e < rope.rot) {
                                const bool second = at.d + e >= half;
                                const int j = second ? at.d + e - half : at.d + e;
                                const float2 cs = turns[t * half + j];
                                y[e] = turn(y[e], cs.x, row[second ? j : j + half], cs.y, second);
                            }
                }
                x[i] = make_float4(y[0], y[1], y[2], y[3]);
            }
        }
        // the largest finite magnitude; not negative, it has the order of its bits
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i)
            top = largest(largest(top, x[i].x, x[i].y), x[i].z, x[i].w);
        const bool new_odd = __any_sync(0xffffffffu, !(top < INFINITY));
        const bool odd = new_odd || (__float_as_uint(was) >> 31) != 0;
        if (new_odd) {
            top = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float m[4] = {fabsf(x[i].x), fabsf(x[i].y), fabsf(x[i].z), fabsf(x[i].w)};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    top = m[e] < INFINITY ? fmaxf(top, m[e]) : top;
            }
        }
        top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
        const float kept = fabsf(was) < INFINITY ? fabsf(was) : 0.0f;  // not written before: anything
        float scale = __fmul_rn(top, 0x1.020408p-7f);  // 1/127
        scale = scale < 0x1p-126f ? 0.0f : scale;
        scale = kept > scale ? kept : scale;
        const float inverse = scale > 0.0f ? __frcp_rn(scale) : 0.0f;
        const bool again = stays && kept != scale;
        const float ratio = again && scale > 0.0f ? __fdiv_rn(kept, scale) : 0.0f;
        int8_t* to = codes + t0 * c.head_dim;
        const int step = at.rows_at_once * c.head_dim;
        if (N > 1 && whole_of(w, src) && !new_odd) {
#pragma unroll
            for (int i = 0; i < N; ++i, to += step)
                if (at.in)
                    *reinterpret_cast<uint32_t*>(to) = codes_of(x[i], inverse);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i, to += step) {
                const int t = t0 + i * at.rows_at_once;
                if (!at.in || t < w.from || t >= w.to)
                    continue;
                uint32_t q = codes_of(x[i], inverse);
                if (new_odd) {
                    const float m[4] = {fabsf(x[i].x), fabsf(x[i].y), fabsf(x[i].z), fabsf(x[i].w)};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!(m[e] < INFINITY))
                            q = (q & ~(0xffu << (8 * e))) | (0x80u << (8 * e));
                }
                *reinterpret_cast<uint32_t*>(to) = q;
            }
        }
        if (again) {
#pragma unroll 4
            for (int t = at.row; t < w.from; t += at.rows_at_once) {
                uint32_t* const stays_at = reinterpret_cast<uint32_t*>(codes + t * c.head_dim);
                if (!at.in)
                    continue;
                const uint32_t old = *stays_at, was_odd = odd_bytes(old);
                const uint32_t q = codes_of(numbers_of(old, 1.0f), ratio);
                *stays_at = (q & ~was_odd) | (0x80808080u & was_odd);
            }
        }
        if (lane == 0)
            *scale_at = odd ? -scale : scale;
        __syncwarp();
    };
    const std::integral_constant<int, STEPS> all{};
    const std::integral_constant<int, 1> one{};
    // the first values, the pages and the angles, none of which needs another
    if (warp < units) {
        if (few_of(item[warp / heads]))
            load(warp, one);
        else
            load(warp, all);
    }
    find_pages(p, count, item);
    if constexpr (TURN != kStill) {
        for (int r = warp; r < count * kBlock; r += kThreads / 32) {
            const Item& w = item[r / kBlock];
            const int t = r % kBlock;
            if (t < w.from || t >= w.to)
                continue;
            const float* const row = angles_of(rope, w.position + t);
            const float nan = __int_as_float(0x7fffffff);
            for (int i = lane; i < half; i += 32)
                angles[r * half + i] = row ? __ldg(reinterpret_cast<const float2*>(row) + i) : make_float2(nan, nan);
        }
    }
    __syncthreads();
    for (int u = warp; u < units; u += kThreads / 32) {
        const Item& w = item[u / heads];
        if (few_of(w)) {
            if (u != warp)
                load(u, one);
            if (w.unit >= 0)
                write(u, one);
        } else {
            if (u != warp)
                load(u, all);
            if (w.unit >= 0)
                write(u, all);
        }
    }
}

struct Sink {
    void* x;
    int64_t token, head;
    int vec;
};

// STEPS: how often the warp moves on in a block's 16 rows; a lane writes 16 bytes of
// each, so that it has 4 codes (for binary32) or 8.
template <typename T, int STEPS>
__global__ void __launch_bounds__(kThreads, 3) read8_kernel(const Params p, const Sink k, const Sink v, const int items)
{
    constexpr int V = 16 / sizeof(T), WORDS = V / 4;
    grid_dependency_launch();
    __shared__ Item item[kMostItems];
    const comp_kv8_cache_t& c = p.cache;
    const int heads = 2 * c.kv_heads, blocks = c.page_size / kBlock;
    const int count = find_items(p, items, item);
    find_pages(p, count, item);
    __syncthreads();
    const Lanes at(c.head_dim, V);
    for (int u = threadIdx.x >> 5; u < count * heads; u += kThreads / 32) {
        const Item& w = item[u / heads];
        const int head = u % heads / 2, is_v = u % 2;
        const Sink& dst = is_v ? v : k;
        const bool there = w.unit >= 0;  // no page, and tokens of no sequence: zeros
        const int64_t unit = there ? w.unit + head : 0;
        const int8_t* const codes = (is_v ? c.v : c.k) + (unit * c.page_size + w.slot) * c.head_dim + at.d;
        const float held = there ? (is_v ? c.v_scale : c.k_scale)[unit * blocks + w.slot / kBlock] : 0.0f;
        T* const to0 = static_cast<T*>(dst.x) + w.token0 * dst.token + head * dst.head + at.d;
        uint32_t q[STEPS][WORDS];
        auto fetch = [&](uint32_t(&f)[WORDS], const int8_t* from) {
            if constexpr (WORDS == 1) {
                f[0] = __ldcs(reinterpret_cast<const uint32_t*>(from));
            } else {
                const uint2 two = __ldcs(reinterpret_cast<const uint2*>(from));
                f[0] = two.x;
                f[1] = two.y;
            }
        };
        auto write = [&](T* to, const float4(&x)[WORDS]) {
            if constexpr (sizeof(T) == 4)
                *reinterpret_cast<float4*>(to) = x[0];
            else
                *reinterpret_cast<uint4*>(to) =
                    make_uint4(pack_h2(__floats2half2_rn(x[0].x, x[0].y)), pack_h2(__floats2half2_rn(x[0].z, x[0].w)),
                               pack_h2(__floats2half2_rn(x[WORDS - 1].x, x[WORDS - 1].y)),
                               pack_h2(__floats2half2_rn(x[WORDS - 1].z, x[WORDS - 1].w)));
        };
        const float scale = fabsf(held);
        const int8_t* from = codes + at.row * c.head_dim;
        T* to = to0 + at.row * dst.token;
        const int step = at.rows_at_once * c.head_dim;
        const int64_t to_step = at.rows_at_once * dst.token;
        // all 16 rows, numbers all of them, to places that vector stores take
        if (w.from == 0 && w.to == kBlock && there && dst.vec && STEPS * at.rows_at_once == kBlock) {
#pragma unroll
            for (int i = 0; i < STEPS; ++i, from += step) {
#pragma unroll
                for (int j = 0; j < WORDS; ++j)
                    q[i][j] = 0;
                if (at.in)
                    fetch(q[i], from);
            }
            if (__float_as_int(held) >= 0) {
#pragma unroll
                for (int i = 0; i < STEPS; ++i, to += to_step) {
                    float4 x[WORDS];
#pragma unroll
                    for (int j = 0; j < WORDS; ++j)
                        x[j] = numbers_of(q[i][j], scale);
                    if (at.in)
                        write(to, x);
                }
                continue;
            }
        } else {
#pragma unroll
            for (int i = 0; i < STEPS; ++i, from += step) {
                const int t = i * at.rows_at_once + at.row;
#pragma unroll
                for (int j = 0; j < WORDS; ++j)
                    q[i][j] = 0;
                if (at.in && t >= w.from && t < w.to && there)
                    fetch(q[i], from);
            }
        }
#pragma unroll
        for (int i = 0; i < STEPS; ++i, to += to_step) {
            const int t = i * at.rows_at_once + at.row;
            if (!at.in || t < w.from || t >= w.to)
                continue;
            float4 x[WORDS];
#pragma unroll
            for (int j = 0; j < WORDS; ++j) {
                x[j] = numbers_of(q[i][j], scale);
                const uint32_t odd = odd_bytes(q[i][j]);
                const float nan = __int_as_float(0x7fffffff);
                x[j] = make_float4(odd & 0xffu ? nan : x[j].x, odd & 0xff00u ? nan : x[j].y,
                                   odd & 0xff0000u ? nan : x[j].z, odd >> 24 ? nan : x[j].w);
            }
            if (dst.vec) {
                write(to, x);
                continue;
            }
#pragma unroll
            for (int j = 0; j < WORDS; ++j) {
                const float y[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if constexpr (sizeof(T) == 4)
                        to[4 * j + e] = y[e];
                    else
                        to[4 * j + e] = __float2half_rn(y[e]);
            }
        }
    }
}

// Blocks for each CTA: as many as give its warps a block of a head each.  131072 tokens of
// one head of 128 are written in 34 us with four blocks a CTA, 47 with two and 84 with one
// (read in 32, 35 and 51).  From three heads on the warps' rounds are not full: 32768
// tokens of three heads take 29 us to write, with four blocks a CTA 24, but 26 and 30 to
// read; 100 sequences of up to 300 new tokens of two heads take 7.0 us as they are, 9.8
// with four.
int items_for(int kv_heads)
{
    return kv_heads >= 4 ? 1 : 4 / kv_heads;
}

template <int STEPS>
void launch_append(const Params& p, const Source& k, const Source& v, const comp_rope_t& r, cudaStream_t s)
{
    const int items = items_for(p.cache.kv_heads);  // their angles are 32 KB at most
    const unsigned grid = static_cast<unsigned>((p.slots + items - 1) / items);
    const size_t smem = static_cast<size_t>(items) * kBlock * r.rot * sizeof(float);
    if (r.rot == 0)
        append8_kernel<STEPS, kStill><<<grid, kThreads, smem, s>>>(p, k, v, r, items);
    else if (r.interleaved)
        append8_kernel<STEPS, kPairs><<<grid, kThreads, smem, s>>>(p, k, v, r, items);
    else if (r.rot % 8 == 0)
        append8_kernel<STEPS, kHalves><<<grid, kThreads, smem, s>>>(p, k, v, r, items);
    else
        append8_kernel<STEPS, kOddHalves><<<grid, kThreads, smem, s>>>(p, k, v, r, items);
}

// Rows of `elem`-byte values that begin on 16 bytes.
int rows_vec(const void* x, int64_t token, int64_t head, int elem)
{
    return aligned16(x) && token % (16 / elem) == 0 && head % (16 / elem) == 0;
}

// The slots of a call; see slot_of_row.  One more for the tokens behind the last
// sequence.  Not more than a grid has CTAs.
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
    if (slots_of(total, rows, cu) > INT32_MAX)
        return COMP_ERR_INVALID_VALUE;
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
    const int items = items_for(cache->kv_heads);
    const unsigned grid = static_cast<unsigned>((p.slots + items - 1) / items);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (elem == 4) {
        if (cache->head_dim > 64)
            read8_kernel<float, 16><<<grid, kThreads, 0, s>>>(p, ks, vs, items);
        else
            read8_kernel<float, 8><<<grid, kThreads, 0, s>>>(p, ks, vs, items);
    } else {
        if (cache->head_dim > 64)
            read8_kernel<__half, 8><<<grid, kThreads, 0, s>>>(p, ks, vs, items);
        else
            read8_kernel<__half, 4><<<grid, kThreads, 0, s>>>(p, ks, vs, items);
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
    if (slots_of(total, rows, cu) > INT32_MAX)
        return COMP_ERR_INVALID_VALUE;
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
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cache->head_dim > 64)
        launch_append<16>(p, ks, vs, r, s);
    else
        launch_append<8>(p, ks, vs, r, s);
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
